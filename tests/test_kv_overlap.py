"""kv_evict's arrays may not overlap, but for the state in place: heads write
new_lens while others still read lens, so one buffer for both would have some of
them skip their eviction.  Refused on the host, before any device is touched (CPU
tests); layouts that share a buffer without sharing a word run (GPU test)."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from tests._kv import HostCache, evict
from tests.test_kv_abi import EVICT, _call, lib  # noqa: F401  (lib: the fixture)

# addresses far apart from each other; never dereferenced
BATCH, HEADS, WIDTH, STATE = 2, 2, 4, 64
APART = {n: 0x100000 * (i + 1) for i, n in enumerate(
    ("table", "lens", "seen", "weights", "positions", "new_lens", "new_weights", "new_positions"))}
ROW = 4 * STATE


def _refused(lib, **over):
    a = dict(APART, batch=BATCH, width=WIDTH, state=STATE)
    a.update(over)
    assert set(a) <= set(EVICT)
    return _call(lib, "kv_evict", **a) == agq.QMV_ERR_UNSUPPORTED and \
        b"overlap" in lib.qmv_kv_last_error()


@pytest.mark.parametrize("read", ["lens", "seen", "table", "weights", "positions"])
@pytest.mark.parametrize("written", ["new_lens", "new_weights", "new_positions"])
def test_a_written_array_over_a_read_one(lib, read, written):
    in_place = {"new_weights": "weights", "new_positions": "positions"}
    if in_place.get(written) != read:
        assert _refused(lib, **{written: APART[read]})
    # by one word from either side, and in the middle
    size = {"lens": 4 * BATCH, "seen": 4 * BATCH, "new_lens": 4 * BATCH, "table": 4 * BATCH * WIDTH}
    state = BATCH * HEADS * ROW
    assert _refused(lib, **{written: APART[read] + size.get(read, state) - 4})
    assert _refused(lib, **{written: APART[read] - size.get(written, state) + 4})


def test_two_written_arrays(lib):
    assert _refused(lib, new_positions=APART["new_weights"])
    assert _refused(lib, new_lens=APART["new_weights"] + 8)
    assert _refused(lib, new_positions=APART["new_lens"] - 3 * ROW)


def test_state_shifted_by_whole_rows(lib):
    # row 1 of the one is row 0 of the other
    assert _refused(lib, new_weights=APART["weights"] + ROW)
    assert _refused(lib, new_positions=APART["positions"] - ROW)


def test_rows_of_a_wider_state(lib):
    # states of 100 words a row, 64 of which are the row's room
    wide = dict(state=100, weights=0x400000)
    assert _refused(lib, **wide, new_weights=0x400000 + 4 * 63)
    assert _refused(lib, **wide, new_weights=0x400000 + 4 * (100 - 63))
    assert _refused(lib, **wide, new_weights=0x400000 - 4 * 63)
    assert _refused(lib, **wide, new_lens=0x400000 + 4 * 63)
    assert _refused(lib, **wide, new_lens=0x400000 + 4 * 99)


def test_binding_says_so(lib):
    cache = agq.KVCache(*[0x10000] * 6, 8, 2, 16, 128, 4, 64)
    p = APART
    with pytest.raises(agq.QmvError, match="new_lens.*lens") as ei:
        agq.kv_evict(cache, p["table"], p["lens"], p["seen"], p["weights"], p["positions"],
                     p["lens"], p["weights"], p["positions"], BATCH, WIDTH, STATE, 32, stream=0)
    assert ei.value.status == agq.QMV_ERR_UNSUPPORTED


@pytest.mark.gpu
def test_arrays_of_one_buffer_that_share_no_word():
    # weights, positions and their new forms as columns of one buffer, and
    # lens, seen and new_lens behind one another in another
    n, budget = 70, 40
    hc = HostCache([n, 50], 2, 64, 8, 64, 16, seed=31, room=80)
    cache, table, lens = hc.device()
    room = hc.width * hc.S
    buf = torch.zeros((2, 2, 4 * room), device="cuda")
    w = np.random.default_rng(1).random((2, 2, room)).astype(np.float32)
    pos = np.broadcast_to(np.arange(room, dtype=np.int32), w.shape)
    buf[..., :room] = torch.from_numpy(w).cuda()
    buf.view(torch.int32)[..., room:2 * room] = torch.from_numpy(pos.copy()).cuda()
    words = torch.cat((lens, lens, torch.full_like(lens, -9)))
    at, step = buf.data_ptr(), 4 * room
    plain = agq.KVCache(*(None if t is None else t.data_ptr() for t in cache.buffers),
                        hc.num_pages, 2, 16, 64, 8, 64)
    agq.kv_evict(plain, table.data_ptr(), words.data_ptr(), words.data_ptr() + 8, at, at + step,
                 words.data_ptr() + 16, at + 2 * step, at + 3 * step, 2, hc.width, 4 * room, budget,
                 8, 4, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert words.tolist() == [n, 50, n, 50, budget, budget]
    for b, m in enumerate((n, 50)):
        for h in range(2):
            _, src = evict(w[b, h], pos[b, h], m, m, budget, 8, 4)
            assert np.array_equal(buf[b, h, 2 * room:2 * room + budget].cpu().numpy(), w[b, h, src])
            got = buf.view(torch.int32)[b, h, 3 * room:3 * room + budget]
            assert np.array_equal(got.cpu().numpy(), pos[b, h, src])
    assert np.array_equal(buf[..., :room].cpu().numpy(), w)
