"""CPU tests of strides that the kv_* binding is given."""
import pytest
import torch

import affine_group_quantized_b200 as agq
from tests._kv_stand_ins import A, D, H, OnDevice, cache_on, runtime


@pytest.fixture
def said():
    with runtime() as r:
        yield r


@pytest.mark.parametrize("stride", [2 ** 61, 2 ** 62, 2 ** 63 - 8, (2 ** 64 - 64) // 6 // 8 * 8])
@pytest.mark.parametrize("name", ["k", "v"])
def test_strides_whose_bytes_pass_64_bits(said, stride, name):
    # rows * stride * 2 would wrap to a small or negative number of bytes
    cache = cache_on([0] * 6)
    small = OnDevice(2 * 4 * H * D, torch.bfloat16, 0)
    kw = {f"{name}_stride": stride}
    k, v = (small, A) if name == "k" else (A, small)
    with pytest.raises(ValueError, match=f"{name}: "):
        agq.kv_read(cache, k, v, A, A, A, 2, 4, 4, stream=0, **kw)
    with pytest.raises(ValueError, match=f"{name}: "):
        agq.kv_append(cache, k, v, A, A, A, 2, 4, 4, stream=0, **kw)


@pytest.mark.parametrize("stride", [-256, -(2 ** 62), 0])
def test_negative_strides_are_refused(said, stride):
    cache = cache_on([0] * 6)
    small = OnDevice(2 * 4 * H * D, torch.bfloat16, 0)
    with pytest.raises((ValueError, agq.QmvError)):
        agq.kv_append(cache, small, A, A, A, A, 2, 4, 4, k_stride=stride, stream=0)
