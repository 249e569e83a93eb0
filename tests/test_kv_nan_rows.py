"""GPU tests of NaN and infinite rows: kv_append writes affine_quantize's bits
for them too."""
import numpy as np
import pytest
import torch

import affine_group_quantized_b200 as agq
from affine_group_quantized_b200 import synth
from tests._kv import BF16_NAN, HostCache
from tests._parity import dev_bf16, host_bits

pytestmark = pytest.mark.gpu

INF, NINF, NNAN = 0x7F80, 0xFF80, 0xFFC1
BIG, NBIG = 0x7F7F, 0xFF7F                      # the largest finite bf16


def _strange_rows(H, D):
    """Rows of ordinary values with every element, half, or one replaced."""
    kinds = [(BF16_NAN,), (NNAN,), (INF,), (NINF,), (BIG,), (NBIG,), (INF, NINF), (BF16_NAN, INF),
             (BF16_NAN, NINF), (BIG, NBIG), (0x0001,), (0x8001,), (0x8000,), (0x7580,)]
    x = synth.normal_bf16((3 * len(kinds), H, D), 51).copy()
    for i, kind in enumerate(kinds):
        fill = np.resize(np.array(kind, np.uint16), D)
        x[3 * i] = fill
        x[3 * i + 1, :, ::2] = fill[: D // 2] if len(kind) == 1 else np.resize(fill, D // 2)
        x[3 * i + 2, :, 5] = kind[0]
    return x


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("D, gs", [(64, 32), (96, 32), (128, 64), (256, 128)])
def test_appended_rows_are_affine_quantizes_bits(bits, D, gs):
    H, page = 2, 16
    x = _strange_rows(H, D)
    T = len(x)
    hc = HostCache([T], H, D, bits, gs, page, seed=52)
    cache, table, lens = hc.device()
    X, Y = dev_bf16(x), dev_bf16(np.ascontiguousarray(x[::-1]))
    zero, starts = (torch.tensor(i, dtype=torch.int32, device="cuda") for i in ([0], [0, T]))
    agq.kv_append(cache, X, Y, table, zero, starts, 1, T, hc.width)
    K, V = torch.empty_like(X), torch.empty_like(Y)
    agq.kv_read(cache, K, V, table, zero, starts, 1, T, hc.width)
    j = torch.arange(T, device="cuda")
    pages, at = table[0].long()[j // page], j % page
    shape = (hc.num_pages, H, page, -1)
    for rows, bufs, back in ((X, (0, 2, 3), K), (Y, (1, 4, 5), V)):
        w = torch.empty((T * H, D * bits // 32), dtype=torch.int32, device="cuda")
        s = torch.empty((T * H, D // gs), dtype=torch.bfloat16, device="cuda")
        b, dense = torch.empty_like(s), torch.empty_like(rows)
        agq.affine_quantize(rows, w, s, b, T * H, D, bits, gs)
        agq.affine_dequantize(w, s, b, dense, T * H, D, bits, gs)
        for buf, want in zip(bufs, (w, s, b)):
            got = cache.buffers[buf].view(shape)[pages, :, at].reshape(want.shape)
            assert np.array_equal(got.view(torch.int16).cpu().numpy(),
                                  want.view(torch.int16).cpu().numpy()), buf
        assert np.array_equal(host_bits(back), host_bits(dense))


def test_a_group_of_nans_has_the_largest_number_as_its_bias():
    H, D, T = 1, 64, 1
    hc = HostCache([T], H, D, 4, 64, 16, seed=53)
    cache, table, lens = hc.device()
    x = dev_bf16(np.full((T, H, D), BF16_NAN, np.uint16))
    agq.kv_append(cache, x, x, table, lens * 0, None, 1, 1, hc.width)
    got = hc.host(cache)
    for name in "kv":
        _, s, b = (a[hc.table[0, 0], 0, 0] for a in got[name])
        assert (s == 0).all() and (b == BIG).all()
