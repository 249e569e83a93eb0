"""CPU tests of the devices that the kv_* binding's arguments lie on."""
import pytest
import torch

import affine_group_quantized_b200 as agq
from tests._kv_stand_ins import OnDevice, cache_on, evict_call, runtime


@pytest.mark.parametrize("at", range(6))
@pytest.mark.parametrize("other", [1, -1])
def test_a_cache_lies_on_one_device(at, other):
    name = ("k", "v", "k_scales", "k_biases", "v_scales", "v_biases")[at]
    devices = [0] * 6
    devices[at] = other
    # the first buffer decides; one on the CPU is refused as such
    match = "CUDA" if other < 0 else f"{'v' if at == 0 else name}: .*device"
    with pytest.raises(ValueError, match=match):
        cache_on(devices)


def test_the_first_tensor_gives_the_device():
    assert cache_on([0] * 6)._device == 0 and cache_on([None] * 6)._device is None
    assert cache_on([None, None, None, 1, 1, None])._device == 1
    with pytest.raises(ValueError, match="v_scales"):
        cache_on([None, None, None, 1, 0, 1])


@pytest.fixture
def said():
    with runtime() as r:
        yield r


def test_tensors_beside_a_cache_of_addresses(said):
    cache = cache_on([None] * 6)
    table = OnDevice(4 * 2 * 4, torch.int32, -1)
    with pytest.raises(ValueError, match="block_table: .*CUDA"):
        evict_call(cache, table)
    table = OnDevice(4 * 2 * 4, torch.int32, 1)       # not where the launch would go
    with pytest.raises(ValueError, match="block_table: .*device"):
        evict_call(cache, table)
    said["device"] = 1
    with pytest.raises(agq.QmvError, match="overlaps"):
        evict_call(cache, table)


def test_tensors_beside_a_cache_of_tensors(said):
    cache = cache_on([0] * 6)
    for d in (-1, 1):
        with pytest.raises(ValueError, match="lens: .*device"):
            evict_call(cache, lens=OnDevice(8, torch.int32, d))
    said["device"] = 1
    with pytest.raises(ValueError, match="current device"):
        evict_call(cache)


def test_scales_of_a_bf16_cache_are_ignored():
    rows = [OnDevice(2 * 8 * 2 * 16 * 128, torch.bfloat16, 0) for _ in range(2)]
    other = OnDevice(4, torch.float16, -1)
    cache = agq.KVCache(*rows, other, other, other, other, 8, 2, 16, 128, 16, 0)
    assert cache._device == 0
