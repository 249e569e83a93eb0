"""Stand-ins for tensors on a GPU and for torch's current device and stream, for
CPU tests of the kv_* binding's checks."""
import contextlib

import torch

import affine_group_quantized_b200 as agq

A = 0x10000  # a fake device address; never dereferenced
H, D, PAGES, PAGE = 2, 128, 8, 16


class Device:
    def __init__(self, index):
        self.index = index


class OnDevice:
    """As much of a tensor as the binding looks at."""

    def __init__(self, nbytes, dtype, device):
        self.nbytes, self.dtype = nbytes, dtype
        self.index = device
        self.is_cuda, self.device = device >= 0, Device(device)

    def numel(self):
        return self.nbytes // self.dtype.itemsize

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return A

    def dim(self):
        return 1


def buffers(devices, bits=4):
    rows = PAGES * H * PAGE
    sizes = [rows * D * bits // 8] * 2 + [2 * rows * D // 64] * 4
    types = [torch.int32] * 2 + [torch.bfloat16] * 4
    return [OnDevice(n, t, d) if d is not None else A for n, t, d in zip(sizes, types, devices)]


def cache_on(devices):
    return agq.KVCache(*buffers(devices), PAGES, H, PAGE, D, 4, 64)


@contextlib.contextmanager
def runtime():
    """The binding's module with functions of the test in place of torch's: what
    they say, and the devices whose streams were asked for."""
    native = agq._kv()
    said = dict(device=0, streams=[])

    def stream(device):
        said["streams"].append(device)
        return 0x5000 + device

    agq._setup(native, lambda: said["device"], stream)
    try:
        yield said
    finally:
        agq._setup(native)


def evict_call(cache, table=A, stream=0, **over):
    # arrays that overlap: the entry point refuses the call after the binding's checks
    args = dict(lens=A, seen=A, weights=A, positions=A, new_lens=A, new_weights=A, new_positions=A)
    args.update(over)
    agq.kv_evict(cache, table, *args.values(), 2, 4, 64, 32, stream=stream)
