"""CPU-only checks of the key-value cache entry points: bad arguments are
refused on the host with the documented status codes, before any device is
touched, and the binding refuses what it can see."""
import ctypes

import pytest

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import build

A = 0x10000  # a 16-byte aligned fake device address; never dereferenced


@pytest.fixture(scope="module")
def lib():
    build.build()
    return agq.lib()


def _cache(**over):
    c = dict(k=A, v=A, k_scales=A, k_biases=A, v_scales=A, v_biases=A, num_pages=8,
             num_kv_heads=2, page_size=16, head_dim=128, bits=4, group_size=64)
    c.update(over)
    return ctypes.byref(agq._KVCacheStruct(**c))


APPEND = dict(cache=None, k=A, v=A, k_stride=256, v_stride=256, table=A, lens=A, starts=A,
              batch=2, tokens=4, width=4, seen=None, positions=None, weights=None, state=0,
              status=None, stream=None)
READ = {n: v for n, v in APPEND.items() if n not in ("seen", "positions", "weights", "state")}
ATTEND = dict(cache=None, q=A, q_stride=512, table=A, lens=A, out=A, batch=2, heads=4, width=4,
              scale=1.0, weights=None, state=0, workspace=A, nbytes=1 << 30, status=None,
              stream=None)
EVICT = dict(cache=None, table=A, lens=A, seen=A, weights=A, positions=A, new_lens=A, new_weights=A,
             new_positions=A, batch=2, width=4, state=64, budget=32, recent=8, sinks=4, status=None,
             stream=None)
CALLS = {"kv_append": APPEND, "kv_read": READ, "kv_attention": ATTEND, "kv_evict": EVICT}


def _call(lib, name, cache=None, **over):
    a = dict(CALLS[name])
    a.update(over)
    a["cache"] = _cache() if cache is None else cache
    return getattr(lib, name)(*a.values())


@pytest.mark.parametrize("name", CALLS)
def test_cache_checks(lib, name):
    def bad(**over):
        return _call(lib, name, cache=_cache(**over))

    assert getattr(lib, name)(None, *list(CALLS[name].values())[1:]) == agq.QMV_ERR_NULL
    assert bad(k=None) == agq.QMV_ERR_NULL
    assert bad(v_biases=None) == agq.QMV_ERR_NULL
    assert name in lib.qmv_kv_last_error().decode()
    for b in (0, 2, 3, 5, 6, 32):
        assert bad(bits=b) == agq.QMV_ERR_UNSUPPORTED
    for d in (0, 32, 80, 192, 512):
        assert bad(head_dim=d) == agq.QMV_ERR_UNSUPPORTED
    assert bad(group_size=16) == agq.QMV_ERR_UNSUPPORTED
    assert bad(head_dim=96) == agq.QMV_ERR_SHAPE            # 64 does not divide 96
    assert bad(head_dim=64, group_size=128) == agq.QMV_ERR_SHAPE
    assert bad(num_pages=0) == agq.QMV_ERR_SHAPE
    assert bad(num_kv_heads=-1) == agq.QMV_ERR_SHAPE
    assert bad(page_size=0) == agq.QMV_ERR_SHAPE
    assert bad(page_size=24) == agq.QMV_ERR_UNSUPPORTED     # not a multiple of 16
    assert bad(num_pages=1 << 27) == agq.QMV_ERR_UNSUPPORTED  # 2^32 rows
    assert bad(v=A + 8) == agq.QMV_ERR_ALIGN
    assert bad(k_scales=A + 2) == agq.QMV_ERR_ALIGN
    # bf16 rows need no scales, and the group size is not looked at
    kw = dict(batch=0)
    if name in ("kv_append", "kv_read"):
        kw["tokens"] = 0
    assert _call(lib, name, cache=_cache(bits=16, k_scales=None, k_biases=None, v_scales=None,
                                         v_biases=None, group_size=0), **kw) == agq.QMV_OK
    assert lib.qmv_kv_last_error() == b""


@pytest.mark.parametrize("name", CALLS)
def test_batch_and_table_checks(lib, name):
    assert _call(lib, name, batch=-1) == agq.QMV_ERR_SHAPE
    assert _call(lib, name, batch=5000) == agq.QMV_ERR_UNSUPPORTED
    assert _call(lib, name, width=0) == agq.QMV_ERR_SHAPE
    assert _call(lib, name, table=None) == agq.QMV_ERR_NULL
    assert _call(lib, name, table=A + 2) == agq.QMV_ERR_ALIGN
    assert _call(lib, name, lens=None) == agq.QMV_ERR_NULL
    assert _call(lib, name, lens=A + 1) == agq.QMV_ERR_ALIGN
    assert _call(lib, name, status=A + 2) == agq.QMV_ERR_ALIGN


@pytest.mark.parametrize("name", ["kv_append", "kv_read"])
def test_row_checks(lib, name):
    assert _call(lib, name, k=None) == agq.QMV_ERR_NULL
    assert _call(lib, name, tokens=-1) == agq.QMV_ERR_SHAPE
    assert _call(lib, name, starts=None, tokens=3) == agq.QMV_ERR_SHAPE  # one per sequence
    assert _call(lib, name, k_stride=255) == agq.QMV_ERR_SHAPE
    assert _call(lib, name, v_stride=260) == agq.QMV_ERR_ALIGN
    assert _call(lib, name, v=A + 2) == agq.QMV_ERR_ALIGN
    assert _call(lib, name, starts=A + 2) == agq.QMV_ERR_ALIGN
    assert _call(lib, name, tokens=0) == agq.QMV_OK          # nothing enqueued


def test_append_state_checks(lib):
    assert _call(lib, "kv_append", seen=A) == agq.QMV_ERR_NULL        # the three go together
    assert _call(lib, "kv_append", seen=A, positions=A, weights=A, state=63) == agq.QMV_ERR_SHAPE
    assert _call(lib, "kv_append", seen=A, positions=A + 2, weights=A, state=64) == agq.QMV_ERR_ALIGN


def test_attention_checks(lib):
    def bad(**over):
        return _call(lib, "kv_attention", **over)

    assert bad(q=None) == agq.QMV_ERR_NULL
    assert bad(out=None) == agq.QMV_ERR_NULL
    assert bad(heads=3) == agq.QMV_ERR_SHAPE                 # two kv heads
    assert bad(heads=0) == agq.QMV_ERR_SHAPE
    assert bad(scale=float("nan")) == agq.QMV_ERR_SHAPE
    assert bad(q_stride=504) == agq.QMV_ERR_SHAPE
    assert bad(q_stride=516) == agq.QMV_ERR_ALIGN
    assert bad(out=A + 8) == agq.QMV_ERR_ALIGN
    assert bad(weights=A, state=63) == agq.QMV_ERR_SHAPE
    assert bad(batch=0) == agq.QMV_OK
    n = ctypes.c_size_t(7)
    w = lib.kv_attention_workspace
    assert w(_cache(), 2, 4, 4, 0, None) == agq.QMV_ERR_NULL
    assert w(_cache(), 2, 3, 4, 0, ctypes.byref(n)) == agq.QMV_ERR_SHAPE
    assert w(_cache(bits=3), 2, 4, 4, 0, ctypes.byref(n)) == agq.QMV_ERR_UNSUPPORTED
    assert n.value == 7


def test_evict_checks(lib):
    def bad(**over):
        return _call(lib, "kv_evict", **over)

    for name in ("seen", "weights", "positions", "new_lens", "new_weights", "new_positions"):
        assert bad(**{name: None}) == agq.QMV_ERR_NULL
        assert bad(**{name: A + 2}) == agq.QMV_ERR_ALIGN
    assert bad(budget=0) == agq.QMV_ERR_SHAPE
    assert bad(recent=-1) == agq.QMV_ERR_SHAPE
    assert bad(recent=30, sinks=4) == agq.QMV_ERR_SHAPE
    assert bad(state=63) == agq.QMV_ERR_SHAPE
    assert bad(width=20000, state=320000) == agq.QMV_ERR_UNSUPPORTED
    assert bad(batch=0) == agq.QMV_OK


def test_binding_raises_with_message(lib):
    cache = agq.KVCache(A, A, A, A, A, A, 8, 2, 16, 128, 7, 64)
    with pytest.raises(agq.QmvError) as ei:
        agq.kv_evict(cache, A, A, A, A, A, A, A, A, 2, 4, 64, 32, stream=0)
    assert ei.value.status == agq.QMV_ERR_UNSUPPORTED and "bits=7" in str(ei.value)


def test_binding_checks_tensors():
    import torch
    with pytest.raises(ValueError, match="k: "):
        agq.KVCache(torch.zeros(8), A, A, A, A, A, 8, 2, 16, 128, 4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        agq.KVCache(torch.zeros(8 * 2 * 16 * 16, dtype=torch.int32), A, A, A, A, A, 8, 2, 16, 128,
                    4, 64)
    cache = agq.KVCache(A, A, A, A, A, A, 8, 2, 16, 128, 4, 64)
    with pytest.raises(ValueError, match="workspace"):
        agq.kv_attention(cache, A, A, A, A, 2, 4, 4, 1.0, None, stream=0)
    t = torch.zeros((4, 128, 2), dtype=torch.bfloat16).transpose(1, 2)
    with pytest.raises(ValueError, match="contiguous"):
        agq.kv_append(cache, t, A, A, A, A, 2, 4, 4, stream=0)
    with pytest.raises(ValueError, match="bf16"):
        agq.kv_append(cache, torch.zeros((4, 2, 128)), A, A, A, A, 2, 4, 4, stream=0)
    with pytest.raises(ValueError, match="block_table"):
        agq.kv_read(cache, A, A, torch.zeros(7, dtype=torch.int32), A, A, 2, 4, 4, stream=0)
