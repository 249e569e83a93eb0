"""The stream of a kv_* call that names none: the current one, on the CPU with
stand-ins, and on the GPU."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from tests._kv import HostCache, attention
from tests._kv_stand_ins import cache_on, evict_call, runtime
from tests._parity import dev_bf16, host_bits


@pytest.fixture
def said():
    with runtime() as r:
        yield r


@pytest.mark.parametrize("devices", [[None] * 6, [0] * 6])
def test_no_stream_is_the_current_one(said, devices):
    # of a cache of plain addresses too: of the current device, where the launch goes
    with pytest.raises(agq.QmvError, match="overlaps"):
        evict_call(cache_on(devices), stream=None)
    assert said["streams"] == [0]
    if devices[0] is None:
        said["device"] = 1
        with pytest.raises(agq.QmvError, match="overlaps"):
            evict_call(cache_on(devices), stream=None)
        assert said["streams"] == [0, 1]
    with pytest.raises(agq.QmvError, match="overlaps"):
        evict_call(cache_on(devices), stream=0x77)
    assert len(said["streams"]) == (2 if devices[0] is None else 1)


@pytest.mark.gpu
def test_a_cache_of_addresses_in_a_captured_graph():
    # captured without naming a stream: the call goes to the capturing one
    hc = HostCache([300, 20], 2, 128, 4, 64, 16, seed=71)
    cache, table, lens = hc.device()
    plain = agq.KVCache(*(t.data_ptr() for t in cache.buffers), hc.num_pages, 2, 16, 128, 4, 64)
    q16 = np.ascontiguousarray(host_bits(torch.randn((2, 8, 128), device="cuda").bfloat16()))
    q = dev_bf16(q16)
    out = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(agq.kv_attention_workspace(plain, 2, 8, hc.width), dtype=torch.uint8, device="cuda")
    ref, bound, _ = attention(hc, q16, 8, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        agq.kv_attention(plain, q, table, lens, out, 2, 8, hc.width, 0.1, ws)
    assert (out == 0).all()
    g.replay()
    torch.cuda.synchronize()
    assert (np.abs(out.float().cpu().numpy() - ref) <= bound).all()
    # and a side stream's events order it
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out.zero_()
        agq.kv_attention(plain, q, table, lens, out, 2, 8, hc.width, 0.1, ws)
    side.synchronize()
    assert (np.abs(out.float().cpu().numpy() - ref) <= bound).all()
