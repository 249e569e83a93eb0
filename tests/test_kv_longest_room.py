"""CPU test of the longest room kv_attention takes: slots, and the ends of tiles and
blocks behind the last one, are numbered in 31 bits."""
import ctypes

import pytest

import affine_group_quantized_b200 as agq
from tests.test_kv_abi import _cache, _call, lib  # noqa: F401  (lib: the fixture)


@pytest.mark.parametrize("page, width", [(16, (1 << 27) - 1), (16, (1 << 27) - 255), (4096, (1 << 19) - 1),
                                         (1 << 20, (1 << 11) - 1)])
@pytest.mark.parametrize("weights", [False, True])
def test_rooms_whose_last_tiles_end_past_31_bits(lib, page, width, weights):
    room = page * width
    cache = dict(page_size=page, num_pages=1, num_kv_heads=1)
    kw = dict(weights=0x10000, state=room) if weights else {}
    past = room > (1 << 31) - 4096
    n = ctypes.c_size_t(0)
    # (refused before a device is looked for; what is taken would need one)
    status = _call(lib, "kv_attention", cache=_cache(**cache), batch=1, heads=1, width=width,
                   q_stride=128, nbytes=0, **kw) if past else None
    if past:
        assert status == agq.QMV_ERR_UNSUPPORTED
        assert b"room" in lib.qmv_kv_last_error()
        assert lib.kv_attention_workspace(_cache(**cache), 1, 1, width, int(weights),
                                          ctypes.byref(n)) == agq.QMV_ERR_UNSUPPORTED
    else:
        assert lib.kv_attention_workspace(_cache(**cache), 1, 1, width, int(weights),
                                          ctypes.byref(n)) != agq.QMV_ERR_UNSUPPORTED
